"""paged_attention_shared_prefix over 8-bit caches whose scales lie outside what the 8-bit
write makes of FP16 rows: zero, subnormal, very small, negative, large and not finite. A
batch of one has its prefix streamed, a larger one takes it to the tensor cores: both
are held to the same 64-bit softmax, with the bounds of serving_plain."""
import numpy as np
import pytest

from serving_plain import E4M3, INT8, AttentionCase
from test_gpu_attention import call, check, tensors

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BATCHES = [1, 40]           # 4 and 160 rows a KV head
FORMATS = [E4M3, INT8]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rope_kv_cache_gb300 import build
    build.build_library()


def make(seed, B, fmt, D=128, P=90, **kw):
    return AttentionCase(seed, B, 1, 8, 2, D, 16, P, [3 + 7 * i % 40 for i in range(B)], fmt, **kw)


def slots(c, plane, which):
    """(page, row) of the prefix positions and of every sequence's own positions whose number
    modulo 5 is in `which`."""
    out = []
    for p in range(c.P):
        if p % 5 in which:
            out.append((int(c.prefix_table[plane, p // c.tpp]) - plane * c.pages, p % c.tpp))
    for b in range(c.B):
        for p in range(c.P, int(c.kv_lens[b])):
            if p % 5 in which:
                out.append((int(c.page_table[b, plane, p // c.tpp]) - plane * c.pages, p % c.tpp))
    return out


def set_scale(c, plane, which, value, head=slice(None)):
    for page, row in slots(c, plane, which):
        c.scales[plane, page, head, row] = value


def run(c):
    t = tensors(c)
    call(c, t)
    check(c, t)


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -149, 2.0 ** -134.8, 2.0 ** -128.5, 2.0 ** -126, 2.0 ** -115,
                                   2.0 ** -101, 2.0 ** -61, 2.0 ** -41, 2.0 ** -33])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B", BATCHES)
def test_small_v_scales_beside_ordinary_ones(B, fmt, scale):
    c = make(900, B, fmt)
    set_scale(c, 1, {1, 3}, scale)
    run(c)


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -149, 2.0 ** -130, 2.0 ** -115, 2.0 ** -80, 2.0 ** -39])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("B", BATCHES)
def test_all_v_scales_small(B, D, scale):
    c = make(910, B, INT8, D=D)
    set_scale(c, 1, {0, 1, 2, 3, 4}, scale)
    run(c)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B", BATCHES)
def test_a_zero_row_of_v_costs_the_others_no_accuracy(B, D, fmt):
    """Tokens with V scale 0 and the largest scores, beside V rows of about 2^-10 with small weights."""
    c = make(920, B, fmt, D=D, P=40, v_scale=2.0 ** -10)
    set_scale(c, 1, {1}, 0.0)
    for page, row in slots(c, 0, {1}):
        c.scales[0, page, :, row] *= 6
    run(c)


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("where", ["prefix", "own"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B", BATCHES)
def test_a_v_scale_that_is_not_finite_leaves_lse_alone(B, fmt, where, value):
    """Only `out` depends on V: the rows that see the token get no finite element, their
    lse and the other heads are as ever."""
    c = make(930, B, fmt)
    p = 7 if where == "prefix" else c.P + 1
    tab = c.prefix_table if where == "prefix" else c.page_table[0]
    c.scales[1, tab[1, p // c.tpp] - c.pages, 1, p % c.tpp] = value
    t = tensors(c)
    call(c, t)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        out, lse, tol_o, tol_l = c.solve()
    got, gl = t["out"].cpu().numpy().astype(np.float64), t["lse"].cpu().numpy().astype(np.float64)
    assert (np.abs(gl - lse) <= tol_l).all()
    hit = np.zeros(got.shape, bool)
    hit[slice(None) if where == "prefix" else 0, :, 4:] = True
    assert not np.isfinite(got[hit]).any()
    assert (np.abs(got[~hit] - out[~hit]) <= tol_o[~hit]).all()


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("B", BATCHES)
def test_a_k_scale_that_is_nan_reaches_out_and_lse(B, value):
    """The scores are not finite (the codes of the token have both signs): no row of that
    head has a result, on either path, and the join passes it on."""
    c = make(940, B, INT8)
    c.scales[0, c.prefix_table[0, 0], 0, 3] = value
    if not np.isnan(value):
        c.pool[0, c.prefix_table[0, 0], 3, 0] = 0            # 0 * infinity
    t = tensors(c)
    call(c, t)
    torch.cuda.synchronize()
    got, gl = t["out"].cpu().numpy(), t["lse"].cpu().numpy()
    assert np.isnan(got[:, :, :4]).all() and np.isnan(gl[:, :, :4]).all()
    assert np.isfinite(got[:, :, 4:]).all() and np.isfinite(gl[:, :, 4:]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B", BATCHES)
def test_negative_and_zero_scales(B, fmt):
    c = make(950, B, fmt)
    for plane in (0, 1):
        for page, row in slots(c, plane, {0, 3}):
            c.scales[plane, page, :, row] *= -1
    set_scale(c, 0, {2}, 0.0)
    run(c)


@pytest.mark.parametrize("scale", [2.0 ** 20, 2.0 ** 59])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B", BATCHES)
def test_large_v_scales(B, fmt, scale):
    """Elements past FP16's range become infinite; a dim whose codes are 0 in all tokens of
    such a scale stays finite."""
    c = make(960, B, fmt)
    set_scale(c, 1, {2}, scale)
    set_scale(c, 1, {4}, 0.0)
    for page, row in slots(c, 1, {2}):
        c.pool[1, page, row, :, :64] = 0
    t = tensors(c)
    call(c, t)
    torch.cuda.synchronize()
    out, lse, _, tol_l = c.solve()
    got, gl = t["out"].cpu().numpy().astype(np.float64), t["lse"].cpu().numpy().astype(np.float64)
    assert (np.abs(gl - lse) <= tol_l).all()
    assert np.isfinite(got[..., :64]).all()
    big = np.abs(out) > scale          # a sum of FP16 weights times codes is off by far less
    assert big.any() and not big[..., :64].any()
    assert np.isinf(got[big]).all() and (np.sign(got) == np.sign(out))[big].all()
