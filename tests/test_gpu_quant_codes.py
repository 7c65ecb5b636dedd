"""rope_write_kv_slot_mapping_quant bit for bit: with M the largest code, codes are the
FP32 product x * (M / max|x|) rounded to the nearest code (ties to the even one), scales
the FP32 quotient max|x| / M; zero heads have scale 0 and codes 0."""
import numpy as np
import pytest

import serving_plain as sp
from serving_plain import E4M3, INT8, NEOX
from test_gpu_serving import quantise

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rope_kv_cache_gb300 import build
    build.build_library()


def nearest_e4m3(x):
    """Codes (uint8) of |x| <= 448, ties to the even code, the sign kept."""
    mag = sp.E4M3_VALUES[:0x7F]                      # 0 .. 448, ascending
    a = np.abs(x).astype(np.float64)
    hi = np.clip(np.searchsorted(mag, a), 1, len(mag) - 1)
    up, down = mag[hi] - a, a - mag[hi - 1]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def unrotated(r):
    """A table that rotates by nothing, so that the head's FP32 values are its FP16 ones."""
    return np.concatenate([np.ones((61, r // 2)), np.zeros((61, r // 2))], 1).astype(np.float32)


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("D,r", [(64, 16), (128, 128), (256, 64)])
def test_codes_and_scales_follow_the_definition(D, r, fmt):
    T, Hq, Hkv = 300, 4, 2
    rng = np.random.Generator(np.random.PCG64(D))
    x = (rng.standard_normal((T, Hq + 2 * Hkv, D)) * 2.0 ** rng.integers(-9, 9, (T, 1, 1))).astype(np.float16)
    # products next to and on the borders between codes
    x[:100, Hq:, 0] = 127 if fmt == INT8 else 448
    x[:100, Hq:, 1:] = rng.integers(-254, 255, (100, 2 * Hkv, D - 1)) / 2
    res = quantise(fmt, (T, Hq, Hkv, D, r, NEOX, 16, True), x=x, seed=D, tab=unrotated(r), bad=False)
    top = np.float32(sp.MAXCODE[fmt])
    for plane in (0, 1):
        y = x[:, Hq + plane * Hkv:Hq + (plane + 1) * Hkv].astype(np.float32)
        amax = np.abs(y).max(-1, keepdims=True)
        u = y * (top / amax)
        assert u.dtype == np.float32
        codes, scales = res["codes"][plane][res["slots"]], res["scales"][plane][res["slots"]]
        want = np.rint(u).astype(np.int8).view(np.uint8) if fmt == INT8 else nearest_e4m3(u)
        zero = u == 0                                # an element -0 keeps its sign in E4M3
        assert np.array_equal(codes[~zero], want[~zero]) and not (codes[zero] & 0x7F).any()
        assert np.array_equal(scales, (amax / top)[..., 0])


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("factor", [1.0, 2.0 ** -110])
def test_zero_heads_have_zero_codes(fmt, factor):
    """Heads of +0 and -0 and heads below 2^-100, of both signs: every code is 0, no bit set."""
    T, Hq, Hkv, D, r = 8, 2, 2, 64, 64
    rng = np.random.Generator(np.random.PCG64(4))
    x = rng.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float16)
    if factor == 1.0:
        x[:, Hq:] = np.where(rng.random((T, 2 * Hkv, D)) < 0.5, 0.0, -0.0)
    else:
        x[:, Hq + Hkv:] = -0.0
    res = quantise(fmt, (T, Hq, Hkv, D, r, NEOX, 4, False), x=x, seed=9, tab=sp.table(61, r) * np.float32(factor), bad=False)
    for plane in (0, 1):
        assert not res["codes"][plane][res["slots"]].any()
        assert not res["scales"][plane][res["slots"]].any()
