"""Calls of paged_attention_shared_prefix that its documentation allows at the edges of its
arguments: queries and unseen tokens that are not finite, lengths of any value, pages of
any size, the same page twice, values at FP16's limit."""
import numpy as np
import pytest

from serving_plain import E4M3, F16, INT8, AttentionCase
from test_gpu_attention import call, check, run, tensors

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ALL = [F16, E4M3, INT8]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rope_kv_cache_gb300 import build
    build.build_library()


@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("B,S", [(1, 2), (3, 3), (30, 2)])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(B, S, fmt):
    c = AttentionCase(1000 + B, B, S, 8, 2, 128, 16, 70, [S + 5 * i % 60 for i in range(B)], fmt)
    t = tensors(c)
    call(c, t)
    first, lse = t["out"].clone(), t["lse"].clone()
    t["q"][0, 0, 1] = float("nan")
    t["q"][B - 1, S - 1, 6] = float("inf")
    call(c, t)
    torch.cuda.synchronize()
    keep = torch.ones(B, S, 8, dtype=torch.bool, device="cuda:0")
    keep[0, 0, 1] = keep[B - 1, S - 1, 6] = False
    assert torch.equal(t["out"][keep], first[keep]) and torch.equal(t["lse"][keep], lse[keep])
    assert torch.isnan(t["out"][~keep]).all() and torch.isnan(t["lse"][~keep]).all()


@pytest.mark.parametrize("plane", [0, 1])
@pytest.mark.parametrize("value", [np.nan, np.inf, 0.0])
@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("B", [2, 30])
def test_scales_that_earlier_rows_do_not_see(B, fmt, value, plane):
    """The last new token has a scale that is not finite: the queries before it do not see it."""
    S = 4
    c = AttentionCase(1010, B, S, 8, 2, 64, 16, 40, [S + 3 * i % 30 for i in range(B)], fmt)
    p = int(c.kv_lens[1]) - 1
    c.scales[plane, c.page_table[1, plane, p // 16] - plane * c.pages, :, p % 16] = value
    t = tensors(c)
    call(c, t)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        out, lse, tol_o, tol_l = c.solve()
    got, gl = t["out"].cpu().numpy().astype(np.float64), t["lse"].cpu().numpy().astype(np.float64)
    keep = np.ones(got.shape, bool)
    if value != 0:
        keep[1, -1] = False
    assert (np.abs(got[keep] - out[keep]) <= tol_o[keep]).all()
    rows = keep.all(-1)
    assert (np.abs(gl[rows] - lse[rows]) <= tol_l[rows]).all()


@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("B,S", [(2, 1), (5, 3), (40, 1)])
def test_lengths_of_any_value(B, S, fmt):
    """Negative and extreme lengths: no row, or all that the table holds."""
    P, cols = 37, 6
    c = AttentionCase(1020, B, S, 8, 2, 128, 16, P, [cols * 16 - P] * B, fmt)
    assert c.page_table.shape[2] == cols
    c.kv_lens[0] = 2 ** 31 - 1
    c.kv_lens[1] = -2 ** 31
    if B > 2:
        c.kv_lens[2], c.kv_lens[3], c.kv_lens[4] = -1, P, P + 1
    run(c)


@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("tpp", [1000, 4096])
@pytest.mark.parametrize("B", [1, 20])
def test_pages_longer_than_everything(B, tpp, fmt):
    run(AttentionCase(1030, B, 2, 8, 2, 64, tpp, 333, [2 + 9 * i % 70 for i in range(B)], fmt))


@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("B", [2, 30])
def test_the_same_page_twice(B, fmt):
    """Prefix and sequences name the same pages again and again."""
    c = AttentionCase(1040, B, 1, 8, 2, 128, 16, 96, [33] * B, fmt)
    c.prefix_table[:, 3:] = c.prefix_table[:, :3]
    c.page_table[:, :, 6] = c.prefix_table[:, 0]
    c.page_table[:, :, 7] = c.prefix_table[:, 0]
    c.page_table[:, :, 8] = c.page_table[:1, :, 8]
    run(c)


@pytest.mark.parametrize("sm_scale", [0.0, -0.3, 1e-38, 1e-6, 40.0])
@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("B", [2, 30])
def test_softmax_scales(B, fmt, sm_scale):
    c = AttentionCase(1050, B, 1, 8, 2, 64, 16, 50, [1 + 3 * i % 40 for i in range(B)], fmt)
    run(c, sm_scale=sm_scale)


@pytest.mark.parametrize("P,Hq,Hkv,D", [(0, 1, 1, 64), (100, 2, 1, 64), (1000, 2, 2, 128)])
def test_the_most_query_tokens(P, Hq, Hkv, D):
    """2^15 query tokens of one sequence; every 911th row against a softmax in 64 bits."""
    import rope_kv_cache_gb300 as rk
    S, tpp = 1 << 15, 64
    N = P + S
    pages = -(-N // tpp)
    gen = torch.Generator(device="cuda:0").manual_seed(P)
    q = torch.randn(1, S, Hq, D, device="cuda:0", generator=gen).half()
    pool = torch.randn(2, pages, tpp, Hkv, D, device="cuda:0", generator=gen).half()
    ids = torch.randperm(pages, device="cuda:0", generator=gen).int()
    table = torch.stack([ids, ids + pages]).contiguous()
    out, lse = torch.empty_like(q), torch.empty(1, S, Hq, device="cuda:0")
    rk.paged_attention_shared_prefix(q, pool, table[:, :-(-P // tpp)].contiguous() if P else None, P, table[None].contiguous(),
                                     torch.tensor([N], dtype=torch.int32, device="cuda:0"), out, lse=lse)
    k, v = (pool[p, ids.long()].reshape(-1, Hkv, D)[:N].double().repeat_interleave(Hq // Hkv, 1) for p in (0, 1))
    for s in list(range(0, S, 911)) + [S - 1]:
        n = P + s + 1
        sc = torch.einsum("hd,nhd->hn", q[0, s].double(), k[:n]) * D ** -0.5
        w = torch.softmax(sc, 1)
        want = torch.einsum("hn,nhd->hd", w, v[:n])
        wv = torch.einsum("hn,nhd->hd", w, v[:n].abs())
        # as serving_plain derives it: scores, weights in FP16, FP32 sums of n terms, one FP16 rounding
        ds = (D + 8) * 2.0 ** -23 * torch.einsum("hd,nhd->hn", q[0, s].double().abs(), k[:n].abs()).max() * D ** -0.5
        rel = 2 * torch.expm1(ds) + 2.0 ** -11 + (2 * n + 40) * 2.0 ** -23
        tol = rel * wv + 2.0 ** -11 * want.abs() + 2.0 ** -24 + 2.0 ** -24 * v.abs().max() * n / torch.exp(
            torch.logsumexp(sc, 1) - sc.max(1).values)[:, None]
        assert ((out[0, s].double() - want).abs() <= tol).all(), s
        ref = torch.logsumexp(sc, 1)
        assert ((lse[0, s].double() - ref).abs() <= ds + (n + 40) * 2.0 ** -23 + 2.0 ** -22 * ref.abs()).all(), s


@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("q_scale", [2.0, 4.0])
@pytest.mark.parametrize("B,P,Hq,D", [(300, 0, 4, 64), (300, 0, 4, 128), (300, 0, 4, 256), (60, 110, 8, 128)])
def test_values_at_the_limit_stay_finite(B, P, Hq, D, q_scale, fmt):
    """All of V is the largest FP16 value in magnitude: so is every mean of it."""
    c = AttentionCase(1060, B, 1, Hq, 4, D, 16, P, [1 + 3 * i % 50 for i in range(B)], fmt, q_scale=q_scale)
    if fmt == F16:
        c.pool[1] = np.where(np.isnan(c.pool[1]), c.pool[1], np.float16(65504))
        c.pool[1, ..., 1::2] *= -1
    else:
        c.pool[1] = 127 if fmt == INT8 else 0x7E
        c.pool[1, ..., 1::2] = -127 if fmt == INT8 else 0xFE
        c.scales[1] = np.where(np.isnan(c.scales[1]), c.scales[1], np.float32(65504 / (127 if fmt == INT8 else 448)))
    t = tensors(c)
    call(c, t)
    torch.cuda.synchronize()
    assert torch.isfinite(t["out"]).all(), int((~torch.isfinite(t["out"])).sum())
    check(c, t)
