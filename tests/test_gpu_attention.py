"""paged_attention_shared_prefix against a plain 64-bit softmax over the
same positions. Every slot that no sequence owns holds NaN (codes and scales)."""
import numpy as np
import pytest

import serving_plain as sp
from serving_plain import E4M3, F16, INT8, AttentionCase

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rope_kv_cache_gb300 import build
    build.build_library()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def tensors(c):
    pool = dev(c.pool)
    if c.fmt == E4M3:
        pool = pool.view(torch.float8_e4m3fn)
    return dict(q=dev(c.q), pool=pool, scales=None if c.scales is None else dev(c.scales),
                prefix=dev(c.prefix_table) if c.P else None, table=dev(c.page_table),
                lens=dev(c.kv_lens), out=torch.full(c.q.shape, float("nan"), dtype=torch.float16, device=DEV),
                lse=torch.full(c.q.shape[:3], float("nan"), device=DEV))


def call(c, t, **kw):
    import rope_kv_cache_gb300 as rk
    kw.setdefault("lse", t["lse"])
    rk.paged_attention_shared_prefix(t["q"], t["pool"], t["prefix"], c.P, t["table"], t["lens"], t["out"],
                                     kv_scales=t["scales"], **kw)


def check(c, t, sm_scale=None):
    torch.cuda.synchronize()
    out, lse, tol_o, tol_l = c.solve(sm_scale)
    got, gl = t["out"].cpu().numpy().astype(np.float64), t["lse"].cpu().numpy().astype(np.float64)
    none = np.isinf(lse)
    assert np.array_equal(np.isneginf(gl), none)
    assert (got[none] == 0).all()
    assert np.isfinite(got).all()
    err = np.abs(got - out)
    assert (err <= tol_o).all(), f"out: worst {float((err / np.maximum(tol_o, 1e-30)).max())} x the bound"
    el = np.abs(gl[~none] - lse[~none])
    assert (el <= tol_l[~none]).all(), f"lse: worst {float((el / tol_l[~none]).max())} x the bound"


def run(c, **kw):
    t = tensors(c)
    call(c, t, **kw)
    check(c, t, kw.get("sm_scale"))
    return t


SHAPES = [
    # B, S, Hq, Hkv, D, tpp, prefix, own lengths
    (1, 1, 1, 1, 64, 1, 0, [1]),
    (1, 1, 4, 4, 128, 16, 1, [1]),
    (2, 1, 8, 2, 64, 16, 15, [1, 40]),
    (3, 1, 8, 2, 128, 16, 16, [1, 16, 17]),
    (3, 1, 8, 1, 128, 64, 0, [200, 1, 63]),
    (5, 1, 10, 2, 64, 7, 33, [3, 9, 1, 77, 14]),
    (4, 1, 16, 2, 256, 32, 70, [5, 300, 64, 1]),
    (2, 1, 32, 8, 128, 64, 1000, [129, 700]),
    (3, 2, 8, 2, 128, 16, 31, [2, 20, 100]),
    (2, 5, 4, 4, 64, 5, 21, [5, 64]),
    (2, 7, 32, 4, 128, 32, 130, [7, 90]),
    (1, 40, 8, 2, 128, 64, 100, [75]),
    (2, 33, 6, 2, 256, 16, 0, [33, 70]),
    (19, 1, 8, 2, 128, 16, 257, list(range(1, 20))),
    (70, 1, 16, 4, 64, 16, 129, [1 + (7 * i) % 50 for i in range(70)]),
    (36, 3, 8, 1, 128, 64, 190, [3 + i for i in range(36)]),
    (40, 1, 16, 2, 256, 64, 321, [1 + i for i in range(40)]),
    (1, 200, 4, 1, 64, 16, 77, [230]),
]


@pytest.mark.parametrize("fmt", [F16, E4M3, INT8])
@pytest.mark.parametrize("idx", range(len(SHAPES)))
def test_shapes(idx, fmt):
    run(AttentionCase(400 + idx, *SHAPES[idx], fmt))


LONG = [
    # enough row tiles that one CTA walks many tiles of the prefix: B, S, Hq, Hkv, D, tpp, prefix
    (25, 200, 8, 8, 64, 16, 1500),
    (40, 250, 4, 4, 128, 64, 1111),
    (38, 256, 2, 2, 256, 32, 705),
    (100, 1, 160, 160, 64, 16, 700),
]


@pytest.mark.parametrize("fmt", [F16, E4M3, INT8])
@pytest.mark.parametrize("idx", range(len(LONG)))
def test_many_prefix_tiles_per_cta(idx, fmt):
    B, S, Hq, Hkv, D, tpp, P = LONG[idx]
    c = AttentionCase(450 + idx, B, S, Hq, Hkv, D, tpp, P, [S + i % 7 for i in range(B)], fmt,
                      q_scale=2.0, unmapped=0.1 if idx == 1 else 0.0)
    # scores that grow along the prefix move the running maximum again and again
    grow = np.linspace(0.2, 4.0, P)
    for p in range(P):
        page = c.prefix_table[0, p // tpp]
        if 0 <= page < c.pages:
            if fmt == F16:
                c.pool[0, page, p % tpp] *= np.float16(grow[p])
            else:
                c.scales[0, page, :, p % tpp] *= np.float32(grow[p])
    t = tensors(c)
    call(c, t)
    torch.cuda.synchronize()
    pick = [0, B // 2, B - 1]
    out, lse, tol_o, tol_l = c.solve(batch=pick)
    got, gl = t["out"].cpu().numpy().astype(np.float64), t["lse"].cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all() and np.isfinite(gl).all()
    err, el = np.abs(got - out)[pick], np.abs(gl - lse)[pick]
    assert (err <= tol_o[pick]).all(), float((err / tol_o[pick]).max())
    assert (el <= tol_l[pick]).all(), float((el / tol_l[pick]).max())


@pytest.mark.parametrize("fmt", [F16, E4M3, INT8])
@pytest.mark.parametrize("B,S,G,D", [(5, 1, 4, 128), (3, 4, 2, 64), (24, 2, 8, 128), (20, 1, 2, 256)])
def test_unmapped_pages_and_inactive_sequences(B, S, G, D, fmt):
    own = [None if i % 4 == 1 else S + 13 * i % 90 for i in range(B)]
    run(AttentionCase(500 + B, B, S, 2 * G, 2, D, 16, 100, own, fmt, unmapped=0.3))


@pytest.mark.parametrize("fmt", [F16, E4M3, INT8])
@pytest.mark.parametrize("B", [4, 40])
def test_peaked_rows_and_spread_scales(B, fmt):
    """Scores up to several hundred, K and V heads between 2^-6 and 2^6."""
    own = [1 + 37 * i % 150 for i in range(B)]
    run(AttentionCase(600 + B, B, 1, 8, 2, 128, 16, 300, own, fmt, q_scale=6.0, spread=6.0))


@pytest.mark.parametrize("v_scale", [2.0 ** -16, 2.0 ** 10])
@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("B", [3, 48])
def test_small_and_large_values(B, fmt, v_scale):
    own = [1 + 11 * i % 80 for i in range(B)]
    run(AttentionCase(700 + B, B, 1, 8, 2, 128, 16, 200, own, fmt, v_scale=v_scale))


@pytest.mark.parametrize("sm_scale", [0.0, -0.3, 1.0])
def test_scale(sm_scale):
    run(AttentionCase(800, 20, 1, 8, 2, 64, 16, 50, [1 + i for i in range(20)], F16), sm_scale=sm_scale)


def test_no_row_sees_anything():
    for P in (0, 40):
        c = AttentionCase(810, 3, 2, 4, 2, 64, 16, P, [None, None, None], F16)
        t = run(c)
        assert (t["out"] == 0).all()


def test_table_shorter_than_the_lengths():
    """Positions past the page table's columns are not seen."""
    c = AttentionCase(820, 3, 1, 8, 2, 128, 16, 20, [30, 100, 5], F16)
    c.page_table = np.ascontiguousarray(c.page_table[:, :, :4])
    run(c)


@pytest.mark.parametrize("fmt", [F16, E4M3])
@pytest.mark.parametrize("S,G", [(4, 2), (3, 8), (9, 8)])
def test_non_finite_values_that_earlier_rows_do_not_see(S, G, fmt):
    """The last new token's V holds an infinity and a NaN: only the last query sees them."""
    c = AttentionCase(830, 2, S, 2 * G, 2, 64, 16, 40, [S + 6, S], fmt)
    b, p = 0, int(c.kv_lens[0]) - 1
    page = c.page_table[b, 1, p // 16] - c.pages
    if fmt == F16:
        c.pool[1, page, p % 16, 0, 5], c.pool[1, page, p % 16, 1, 7] = np.inf, np.nan
    else:
        c.pool[1, page, p % 16, 0, 5], c.pool[1, page, p % 16, 1, 7] = 0x7F, 0xFF
    t = tensors(c)
    call(c, t)
    torch.cuda.synchronize()
    got = t["out"].cpu().numpy().astype(np.float64)
    if fmt == F16:
        assert np.isposinf(got[0, -1, :G, 5]).all()
    else:
        assert np.isnan(got[0, -1, :G, 5]).all()
    assert np.isnan(got[0, -1, G:, 7]).all()
    c.pool[1, page, p % 16, 0, 5] = c.pool[1, page, p % 16, 1, 7] = 0      # finite for the reference
    out, _, tol, _ = c.solve()
    keep = np.ones(got.shape, bool)
    keep[0, -1, :G, 5] = keep[0, -1, G:, 7] = False
    assert (np.abs(got - out)[keep] <= tol[keep]).all()


def test_poisoned_scale_reaches_the_rows_that_see_it():
    c = AttentionCase(840, 2, 1, 4, 2, 64, 16, 16, [9, 9], INT8)
    p = 20
    page = c.page_table[1, 1, p // 16] - c.pages
    c.scales[1, page, 0, p % 16] = np.nan
    t = tensors(c)
    call(c, t)
    torch.cuda.synchronize()
    got = t["out"].cpu().numpy()
    assert np.isnan(got[1, 0, :2]).all() and np.isfinite(got[1, 0, 2:]).all() and np.isfinite(got[0]).all()


@pytest.mark.parametrize("B,fmt", [(6, F16), (40, E4M3)])
def test_repeated_calls_are_equal_and_streams_and_graphs_work(B, fmt):
    own = [1 + 29 * i % 120 for i in range(B)]
    c = AttentionCase(850, B, 1, 8, 2, 128, 16, 500, own, fmt)
    t = run(c)
    first, lse = t["out"].clone(), t["lse"].clone()
    import rope_kv_cache_gb300 as rk
    for _ in range(3):
        t["out"].fill_(float("nan"))
        call(c, t)
        assert torch.equal(t["out"], first) and torch.equal(t["lse"], lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t["out"].fill_(float("nan"))
    torch.cuda.synchronize()
    call(c, t, stream=side)
    side.synchronize()
    assert torch.equal(t["out"], first)
    size = rk.paged_attention_workspace_size(t["q"], t["pool"], t["prefix"], c.P, t["table"],
                                             kv_scales=t["scales"])
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    t["out"].fill_(float("nan"))
    call(c, t, workspace=ws, lse=None)
    assert torch.equal(t["out"], first)
    with pytest.raises(rk.RopeKVError):
        call(c, t, workspace=ws[:size - 16])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c, t)
    c2 = AttentionCase(851, B, 1, 8, 2, 128, 16, 500, own, fmt)
    t2 = tensors(c2)
    for n in ("q", "pool", "scales", "prefix", "table", "lens"):
        if t[n] is not None:
            t[n].view(torch.uint8).copy_(t2[n].view(torch.uint8))
    g.replay()
    check(c2, t)


def test_rows_are_independent_of_the_batch():
    """Without a prefix a sequence's result does not depend on its neighbours."""
    c = AttentionCase(860, 5, 1, 8, 2, 128, 16, 0, [50, 3, 120, 1, 77], F16)
    t = run(c)
    import rope_kv_cache_gb300 as rk
    for b in range(5):
        out = torch.zeros(1, 1, 8, 128, dtype=torch.float16, device=DEV)
        rk.paged_attention_shared_prefix(t["q"][b:b + 1], t["pool"], None, 0, t["table"][b:b + 1].contiguous(),
                                         t["lens"][b:b + 1].clone(), out)
        assert torch.allclose(out[0].float(), t["out"][b].float(), rtol=2.0 ** -9, atol=2.0 ** -12)


@pytest.mark.parametrize("fmt", [F16, INT8])
def test_decode_step_end_to_end(fmt):
    """A decode step as it is used: the new token of every sequence is rotated and written
    through its slot, then attended to together with the shared prefix."""
    import rope_kv_cache_gb300 as rk
    B, Hq, Hkv, D, tpp, P = 6, 8, 2, 128, 16, 40
    own = [1 + 9 * i for i in range(B)]
    c = AttentionCase(870, B, 1, Hq, Hkv, D, tpp, P, own, fmt)
    # one page id for both planes, as slots name them
    rng = np.random.Generator(np.random.PCG64(1))
    perm = rng.permutation(c.pages)
    at = 0
    for tab in [c.prefix_table] + list(c.page_table):
        for col in range(tab.shape[1]):
            if tab[0, col] >= 0:
                tab[0, col], tab[1, col] = perm[at], perm[at] + c.pages
                at += 1
    x = rng.standard_normal((2, c.pages, tpp, Hkv, D))
    if fmt == F16:
        c.pool = x.astype(np.float16)
    else:
        c.scales = (np.abs(x).max(-1) / 127).astype(np.float32).transpose(0, 1, 3, 2).copy()
        c.pool = np.rint(x / c.scales.transpose(0, 1, 3, 2)[..., None].astype(np.float64)).astype(np.int8)
    t = tensors(c)
    qkv = rng.standard_normal((B, Hq + 2 * Hkv, D)).astype(np.float16)
    pos = c.kv_lens.astype(np.int64) - 1
    slots = np.array([int(c.page_table[b, 0, pos[b] // tpp]) * tpp + pos[b] % tpp for b in range(B)])
    cs = sp.table(400, D)
    d = dev(qkv)
    q, k, v = d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:]
    q_out = torch.zeros(B, Hq, D, dtype=torch.float16, device=DEV)
    if fmt == F16:
        rk.rope_write_kv_mrope(dev(cs), dev(np.stack([pos] * 3)), rk.mrope_freq_axis([16, 24, 24]), q, k, v,
                               dev(slots), t["pool"][0], t["pool"][1], q_out)
    else:
        rk.rope_write_kv_slot_mapping_quant(dev(cs), dev(pos), q, k, v, dev(slots), t["pool"][0], t["pool"][1],
                                            t["scales"][0], t["scales"][1], q_out)
    t["q"] = q_out.view(B, 1, Hq, D)
    call(c, t)
    torch.cuda.synchronize()
    # the reference sees the cache as the write left it; the write itself is tested elsewhere,
    # here the new rows are the rotated ones
    c.q = q_out.view(B, 1, Hq, D).cpu().numpy()
    c.pool = t["pool"].cpu().numpy()
    if fmt != F16:
        c.scales = t["scales"].cpu().numpy()
    row = cs[pos].astype(np.float64)
    yk, _ = sp.rotate(qkv[:, Hq:Hq + Hkv].astype(np.float64), row[:, :D // 2], row[:, D // 2:], D, sp.NEOX)
    new = c.values()[0].reshape(-1, Hkv, D)[slots]
    assert np.abs(new - yk).max() < (2.0 ** -9 if fmt == F16 else np.abs(yk).max() / 127)
    check(c, t)
