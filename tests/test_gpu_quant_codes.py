"""Codes and scales of rope_write_kv_slot_mapping_quant, bit for bit."""
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
