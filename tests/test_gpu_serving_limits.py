"""The serving operators at head counts that leave warps idle, at large batches, with
pools, rows and strides whose element offsets pass 2^32, and in calls that overlap."""
import numpy as np
import pytest

import serving_plain as sp
from serving_plain import E4M3, F16, INT8, AttentionCase
from test_gpu_attention import call, check, dev, run, tensors

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rope_kv_cache_gb300 import build
    build.build_library()


def need(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of free device memory")


HEADS = [
    # Hkv, G, D, B, S
    (3, 4, 128, 4, 1),
    (5, 2, 64, 20, 1),
    (7, 1, 128, 30, 1),
    (11, 3, 64, 6, 2),
    (13, 1, 256, 3, 1),
    (16, 2, 128, 9, 1),
    (24, 1, 64, 12, 3),
    (17, 8, 64, 2, 5),
]


@pytest.mark.parametrize("fmt", [F16, E4M3, INT8])
@pytest.mark.parametrize("idx", range(len(HEADS)))
def test_head_counts(idx, fmt):
    Hkv, G, D, B, S = HEADS[idx]
    own = [None if i == 2 else S + 17 * i % 71 for i in range(B)]
    run(AttentionCase(900 + idx, B, S, Hkv * G, Hkv, D, 16, 75, own, fmt))


@pytest.mark.parametrize("fmt", [F16, INT8])
@pytest.mark.parametrize("B,P", [(700, 0), (1500, 33), (520, 100)])
def test_many_sequences(B, P, fmt):
    own = [None if i % 7 == 3 else 1 + i % 5 for i in range(B)]
    own[B // 2] = 400
    run(AttentionCase(920 + B, B, 1, 4, 2, 64, 16, P, own, fmt))


def spread_pool(c, pages):
    """The case's pool inside one of `pages` pages, its own pages spread to the very end."""
    at = np.linspace(0, pages - 1, c.pages).astype(np.int64)
    big = torch.zeros((2, pages) + c.pool.shape[2:], dtype={F16: torch.float16, INT8: torch.int8}[c.fmt], device=DEV)
    big[:, at] = dev(c.pool)
    scales = None
    if c.scales is not None:
        scales = torch.zeros((2, pages) + c.scales.shape[2:], device=DEV)
        scales[:, at] = dev(c.scales)

    def move(tab):
        out = np.full_like(tab, -1)
        for plane in (0, 1):
            ids = tab[..., plane, :] - plane * c.pages
            ok = tab[..., plane, :] >= 0
            out[..., plane, :][ok] = at[ids[ok]] + plane * pages
        return out
    return big, scales, move


@pytest.mark.parametrize("fmt", [F16, INT8])
@pytest.mark.parametrize("B", [3, 24])
def test_pool_past_32_bits(B, fmt):
    need(24)
    c = AttentionCase(940, B, 1, 32, 8, 128, 64, 200, [1 + 23 * i % 150 for i in range(B)], fmt)
    t = run(c)
    big, scales, move = spread_pool(c, 40000)
    assert big.numel() > 2 ** 32
    u = dict(t, pool=big, scales=scales, prefix=dev(move(c.prefix_table)), table=dev(move(c.page_table)),
             out=torch.full_like(t["out"], float("nan")), lse=torch.full_like(t["lse"], float("nan")))
    call(c, u)
    assert torch.equal(u["out"], t["out"]) and torch.equal(u["lse"], t["lse"])
    # and read back: the same rows through either table
    import rope_kv_cache_gb300 as rk
    pos = torch.arange(200, 200 + 100, dtype=torch.int32, device=DEV)
    seq = (torch.arange(100, device=DEV) % B).int()
    got = []
    for x in (t, u):
        ko, vo = torch.zeros(100, 8, 128, dtype=torch.float16, device=DEV), torch.zeros(100, 8, 128, dtype=torch.float16, device=DEV)
        rk.paged_kv_read(x["pool"], x["table"], pos, seq, ko, vo, kv_scales=x["scales"])
        got += [ko.view(torch.int16), vo.view(torch.int16)]
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])


def test_read_output_past_32_bits():
    need(24)
    import rope_kv_cache_gb300 as rk
    N, Hkv, D, tpp, pages = 2 ** 22 + 77, 8, 128, 64, 50
    pool = torch.randn(2, pages, tpp, Hkv, D, device=DEV).half()
    table = torch.stack([torch.arange(pages), torch.arange(pages) + pages]).int()[None].to(DEV)
    pos = (torch.arange(N, device=DEV) % (pages * tpp)).int()
    ko = torch.zeros(N, Hkv, D, dtype=torch.float16, device=DEV)
    vo = torch.zeros_like(ko)
    rk.paged_kv_read(pool, table, pos, torch.zeros_like(pos), ko, vo)
    for lo in (0, N // 2, N - 500):
        p = pos[lo:lo + 500].long()
        assert torch.equal(ko[lo:lo + 500], pool[0].view(-1, Hkv, D)[p])
        assert torch.equal(vo[lo:lo + 500], pool[1].view(-1, Hkv, D)[p])


@pytest.mark.parametrize("op", ["mrope", "quant"])
def test_write_past_32_bits(op):
    """Slots behind element 2^32 of the cache, token strides of 2^31 elements."""
    need(40)
    import rope_kv_cache_gb300 as rk
    T, Hq, Hkv, D, bs, blocks = 3, 8, 8, 128, 64, 70000
    stride = 2 ** 31
    x = torch.zeros(2 * stride + (Hq + 2 * Hkv) * D, dtype=torch.float16, device=DEV)
    rows = x.as_strided((T, Hq + 2 * Hkv, D), (stride, D, 1))
    rows.copy_(torch.randn(T, Hq + 2 * Hkv, D, device=DEV))
    tab, pos = dev(sp.table(50, D)), torch.tensor([3, 49, 7], device=DEV)
    far = torch.tensor([blocks * bs - 1, 5, blocks * bs - 700], device=DEV)
    near = torch.tensor([0, 1, 2], device=DEV)
    got = []
    for q, slots, n in ((rows, far, blocks), (rows.contiguous(), near, 1)):
        a, k, v = q[:, :Hq], q[:, Hq:Hq + Hkv], q[:, Hq + Hkv:]
        qo = torch.zeros(T, Hq, D, dtype=torch.float16, device=DEV)
        dt = torch.float16 if op == "mrope" else torch.int8
        kc, vc = torch.zeros(n, bs, Hkv, D, dtype=dt, device=DEV), torch.zeros(n, bs, Hkv, D, dtype=dt, device=DEV)
        ks, vs = torch.zeros(n, Hkv, bs, device=DEV), torch.zeros(n, Hkv, bs, device=DEV)
        if op == "mrope":
            rk.rope_write_kv_mrope(tab, torch.stack([pos, pos.flip(0)]), rk.mrope_freq_axis([D // 4, D // 4]),
                                   a, k, v, slots, kc, vc, qo)
        else:
            rk.rope_write_kv_slot_mapping_quant(tab, pos, a, k, v, slots, kc, vc, ks, vs, qo)
        flat = lambda s: s.transpose(1, 2).reshape(-1, Hkv)[slots]
        got.append((qo, kc.view(-1, Hkv, D)[slots], vc.view(-1, Hkv, D)[slots], flat(ks), flat(vs)))
        assert got[-1][1].any() and got[-1][2].any()
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_query_rows_past_32_bits():
    """2^25 query rows of 128: every sequence has its token and the prefix."""
    need(120)
    import rope_kv_cache_gb300 as rk
    B, H, D, P = 2 ** 18, 128, 128, 20
    q = torch.empty(B, 1, H, D, dtype=torch.float16, device=DEV).normal_()
    pool = torch.randn(2, 8, 16, 1, D, device=DEV).half()
    prefix = torch.tensor([[0, 1], [8, 9]], dtype=torch.int32, device=DEV)
    table = torch.full((B, 2, 2), -1, dtype=torch.int32, device=DEV)
    own = (2 + torch.arange(B, device=DEV) % 6).int()
    table[:, 0, 1], table[:, 1, 1] = own, own + 8
    lens = (P + 1 + torch.arange(B, device=DEV) % 9).int()
    out = torch.zeros_like(q)
    rk.paged_attention_shared_prefix(q, pool, prefix, P, table, lens, out)
    for lo in (0, B // 2 - 1, B - 3):
        for b in range(lo, lo + 3):
            n = int(lens[b])
            pages = [0] + ([int(own[b])] if n > P else [])
            k = torch.cat([pool[0, 0, :, 0], pool[0, 1, :4, 0], pool[0, pages[-1], 4:4 + n - P, 0]]).double()
            v = torch.cat([pool[1, 0, :, 0], pool[1, 1, :4, 0], pool[1, pages[-1], 4:4 + n - P, 0]]).double()
            want = torch.softmax(q[b, 0].double() @ k.T * D ** -0.5, -1) @ v
            # weights in FP16 (2^-11), the result in FP16 (2^-11), scores of FP32 sums
            bound = 3 * 2.0 ** -11 * torch.softmax(q[b, 0].double() @ k.T * D ** -0.5, -1) @ v.abs() + 2.0 ** -14
            assert ((out[b, 0].double() - want).abs() <= bound).all(), b


@pytest.mark.parametrize("fmt", [F16, E4M3])
def test_calls_on_two_streams_at_once(fmt):
    cases = [AttentionCase(960 + i, 40, 1, 8, 2, 128, 16, 700, [1 + 31 * j % 90 for j in range(40)], fmt)
             for i in range(2)]
    ts = [run(c) for c in cases]
    want = [t["out"].clone() for t in ts]
    for t in ts:
        t["out"].zero_()
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in ts]
    for _ in range(20):
        for c, t, s in zip(cases, ts, side):
            call(c, t, stream=s)
    torch.cuda.synchronize()
    for t, w in zip(ts, want):
        assert torch.equal(t["out"], w)


def test_write_attend_write_on_one_stream():
    """Launches that may start early still wait: the pool that one call reads is changed
    before and after it on the same stream, over and over."""
    import rope_kv_cache_gb300 as rk
    B, Hq, Hkv, D, tpp, P = 40, 8, 2, 128, 16, 300
    c = AttentionCase(970, B, 1, Hq, Hkv, D, tpp, P, [1 + i for i in range(B)], INT8)
    t = tensors(c)
    call(c, t)
    check(c, t)
    first = t["out"].clone()
    slots = torch.arange(c.pages * tpp, device=DEV)
    T = len(slots)
    rng = torch.Generator(device=DEV).manual_seed(1)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=rng, device=DEV).half()
    tab, pos = dev(sp.table(64, D)), slots % 64
    qo = torch.zeros(T, Hq, D, dtype=torch.float16, device=DEV)
    pool, scales = t["pool"].clone(), t["scales"].clone()

    def write():
        rk.rope_write_kv_slot_mapping_quant(tab, pos, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], slots,
                                            t["pool"][0], t["pool"][1], t["scales"][0], t["scales"][1], qo)
    write()
    call(c, t)
    second = t["out"].clone()
    assert not torch.equal(first, second)
    outs = []
    for _ in range(10):
        t["pool"].copy_(pool), t["scales"].copy_(scales)
        call(c, t)
        outs.append(t["out"].clone())
        write()
        call(c, t)
        write()
        outs.append(t["out"].clone())
    for i, o in enumerate(outs):
        assert torch.equal(o, second if i % 2 else first), i


def test_sequences_that_share_their_own_pages():
    c = AttentionCase(980, 24, 1, 8, 2, 64, 16, 40, [30] * 24, F16)
    c.page_table[1:] = c.page_table[:1]
    c.q[1:] = c.q[:1]
    t = run(c)
    # equal rows of one batch: equal up to where the work is cut
    assert (t["out"].float() - t["out"][:1].float()).abs().max() <= 2.0 ** -9 * t["out"].float().abs().max()


@pytest.mark.parametrize("fmt", [F16, E4M3])
@pytest.mark.parametrize("B,S", [(6, 1), (40, 1), (12, 3)])
def test_queries_of_inactive_sequences_hold_anything(B, S, fmt):
    own = [None if i % 3 == 1 else S + 19 * i % 60 for i in range(B)]
    c = AttentionCase(990 + B, B, S, 8, 2, 128, 16, 90, own, fmt)
    t = tensors(c)
    idle = [i for i in range(B) if own[i] is None]
    t["q"][idle[::2]] = float("nan")
    t["q"][idle[1::2]] = float("inf")
    call(c, t)
    check(c, t)


def test_result_in_place_of_the_queries():
    c = AttentionCase(1000, 30, 1, 8, 2, 128, 16, 200, [1 + 7 * i % 40 for i in range(30)], F16)
    t = tensors(c)
    call(c, t)
    want = t["out"].clone()
    t["out"] = t["q"]
    call(c, t)
    assert torch.equal(t["q"], want)


@pytest.mark.parametrize("B", [6, 40])
def test_table_wider_than_the_lengths(B):
    """Columns that no sequence reaches change the split of the work, not the result."""
    own = [1 + 5 * i % 70 for i in range(B)]
    c = AttentionCase(1010 + B, B, 1, 8, 2, 128, 16, 700, own, F16)
    c.page_table = np.ascontiguousarray(np.concatenate(
        [c.page_table, np.full((B, 2, 3000), -1, np.int32)], -1))
    run(c)


@pytest.mark.parametrize("seed", range(24))
def test_random_calls(seed):
    """Sizes drawn over the whole range, the workspace guarded by bytes behind its end."""
    import rope_kv_cache_gb300 as rk
    rng = np.random.Generator(np.random.PCG64(2000 + seed))
    pick = lambda *x: x[rng.integers(len(x))]
    log = lambda a, b: int(round(np.exp(rng.uniform(np.log(a), np.log(b)))))
    D, Hkv, G, S = pick(64, 128, 256), pick(1, 2, 3, 4, 5, 8, 9), pick(1, 2, 3, 4, 7, 8, 16), pick(1, 1, 1, 2, 5, 8, 16)
    P, tpp, fmt, B = pick(0, log(1, 60), log(16, 1500)), pick(1, 3, 8, 16, 24, 64, 100), pick(F16, E4M3, INT8), log(1, 40)
    own = [None if rng.random() < 0.1 else S + int(rng.integers(log(1, 300))) for _ in range(B)]
    c = AttentionCase(3000 + seed, B, S, Hkv * G, Hkv, D, tpp, P, own, fmt, q_scale=pick(0.3, 1.0, 3.0),
                      unmapped=pick(0, 0, 0.2), spread=pick(0, 0, 3))
    t = tensors(c)
    size = rk.paged_attention_workspace_size(t["q"], t["pool"], t["prefix"], c.P, t["table"], kv_scales=t["scales"])
    ws = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    call(c, t, workspace=ws[:size])
    check(c, t)
    assert (ws[size:] == 0xFF).all()
