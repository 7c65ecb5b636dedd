"""Refusals of the serving operators' Python binding, each by its own message: every case
differs from a call that would be fine on a GPU in the one argument that is named (the
fine call itself is refused for its CPU tensors, after all shapes have been checked)."""
import pytest

torch = pytest.importorskip("torch")

import rope_kv_cache_gb300 as rk
from rope_kv_cache_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def h(*s):
    return torch.zeros(*s, dtype=torch.float16)


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def i64(*s):
    return torch.zeros(*s, dtype=torch.int64)


def attention(**kw):
    a = dict(q=h(3, 1, 4, 64), pool=h(2, 4, 16, 2, 64), prefix=i32(2, 1), P=16, table=i32(3, 2, 2), lens=i32(3),
             out=h(3, 1, 4, 64), lse=torch.zeros(3, 1, 4), scales=None, scale=None, workspace=None)
    a.update(kw)
    rk.paged_attention_shared_prefix(a["q"], a["pool"], a["prefix"], a["P"], a["table"], a["lens"], a["out"],
                                     lse=a["lse"], kv_scales=a["scales"], sm_scale=a["scale"],
                                     workspace=a["workspace"])


EIGHT = dict(pool=torch.zeros(2, 4, 16, 2, 64, dtype=torch.int8))


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "expected a CUDA device"),
    (dict(lse=None, prefix=None, P=0), ValueError, "expected a CUDA device"),
    (dict(EIGHT, scales=torch.zeros(2, 4, 2, 16)), ValueError, "expected a CUDA device"),
    (dict(lens=i32(2)), ValueError, "kv_lens"),
    (dict(lens=i32(3, 1)), ValueError, "kv_lens"),
    (dict(out=h(3, 1, 2, 64)), ValueError, "kv_lens .* out"),
    (dict(out=h(3, 4, 64)), ValueError, "kv_lens .* out"),
    (dict(lse=torch.zeros(3, 4)), ValueError, "kv_lens .* lse"),
    (dict(lse=torch.zeros(3, 1, 3)), ValueError, "kv_lens .* lse"),
    (dict(q=h(2, 1, 4, 64)), ValueError, "q does not match"),
    (dict(q=h(3, 1, 4, 128)), ValueError, "q does not match"),
    (dict(q=h(3, 4, 64)), ValueError, r"q \[B, S, Hq, D\]"),
    (dict(table=i32(3, 1, 2)), ValueError, "page_table"),
    (dict(table=i32(3, 2)), ValueError, "page_table"),
    (dict(pool=h(1, 4, 16, 2, 64)), ValueError, "page_table"),
    (dict(prefix=i32(1, 1)), ValueError, "prefix_table"),
    (dict(prefix=i32(2)), ValueError, "prefix_table"),
    (dict(EIGHT), ValueError, "kv_scales .* expected"),
    (dict(EIGHT, scales=torch.zeros(2, 4, 16, 2)), ValueError, "kv_scales .* expected"),
    (dict(scales=torch.zeros(2, 4, 2, 16)), ValueError, "no kv_scales"),
    (dict(pool=torch.zeros(2, 4, 16, 2, 64)), TypeError, "kv_cache: dtype Float"),
    (dict(P=2 ** 40), ValueError, "prefix_len is too large"),
    (dict(P=None), TypeError, "NoneType"),
    (dict(scale="1"), TypeError, "real number"),
    (dict(lens=[1, 2, 3]), TypeError, "kv_lens must be a torch.Tensor"),
    (dict(workspace=5), TypeError, "workspace must be a torch.Tensor"),
])
def test_attention(kw, error, match):
    with pytest.raises(error, match=match):
        attention(**kw)


@pytest.mark.parametrize("kw,match", [
    (dict(table=i32(3, 1, 2)), "page_table"),
    (dict(q=h(2, 1, 4, 64)), "q does not match"),
    (dict(prefix=i32(1, 1)), "prefix_table"),
    (dict(EIGHT), "kv_scales"),
])
def test_workspace_size(kw, match):
    a = dict(q=h(3, 1, 4, 64), pool=h(2, 4, 16, 2, 64), prefix=i32(2, 1), table=i32(3, 2, 2))
    assert rk.paged_attention_workspace_size(a["q"], a["pool"], a["prefix"], 16, a["table"]) > 0
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        rk.paged_attention_workspace_size(a["q"], a["pool"], a["prefix"], 16, a["table"])


def test_workspace_size_of_refused_sizes():
    with pytest.raises(rk.RopeKVError):          # a prefix longer than its table
        rk.paged_attention_workspace_size(h(3, 1, 4, 64), h(2, 4, 16, 2, 64), i32(2, 1), 17, i32(3, 2, 2))


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "expected a CUDA device"),
    (dict(pos=i32(4)), ValueError, "row_positions"),
    (dict(k=h(5, 2, 128)), ValueError, "k_out, v_out"),
    (dict(v=h(4, 2, 64)), ValueError, "k_out, v_out"),
    (dict(table=i32(3, 3, 2)), ValueError, "page_table"),
    (dict(scales=torch.zeros(2, 4, 2, 16)), ValueError, "no kv_scales"),
    (dict(EIGHT, scales=torch.zeros(2, 4, 2, 8)), ValueError, "kv_scales .* expected"),
])
def test_read(kw, error, match):
    a = dict(pool=h(2, 4, 16, 2, 64), table=i32(3, 2, 2), pos=i32(5), seq=i32(5), k=h(5, 2, 64), v=h(5, 2, 64), scales=None)
    a.update(kw)
    with pytest.raises(error, match=match):
        rk.paged_kv_read(a["pool"], a["table"], a["pos"], a["seq"], a["k"], a["v"], kv_scales=a["scales"])


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "expected a CUDA device"),
    (dict(kc=torch.zeros(2, 16, 2, 64, dtype=torch.int8), vc=torch.zeros(2, 16, 2, 128, dtype=torch.int8)), ValueError, "inconsistent"),
    (dict(v=h(3, 1, 64)), ValueError, "inconsistent"),
    (dict(qo=h(3, 2, 64)), ValueError, "inconsistent"),
    (dict(slots=i64(2)), ValueError, "inconsistent"),
    (dict(pos=i64(2)), ValueError, "inconsistent"),
    (dict(ks=torch.zeros(2, 16, 2)), ValueError, "key_scales"),
    (dict(vs=torch.zeros(2, 2, 8)), ValueError, "key_scales, value_scales"),
    (dict(kc=h(2, 16, 2, 64)), TypeError, "key_cache: dtype Half"),
    (dict(cs=torch.zeros(64)), ValueError, "cos_sin"),
])
def test_quantised_write(kw, error, match):
    e = lambda: torch.zeros(2, 16, 2, 64, dtype=torch.int8)
    a = dict(cs=torch.zeros(16, 64), pos=i64(3), q=h(3, 4, 64), k=h(3, 2, 64), v=h(3, 2, 64), slots=i64(3), kc=e(),
             vc=e(), ks=torch.zeros(2, 2, 16), vs=torch.zeros(2, 2, 16), qo=h(3, 4, 64), style=rk.NEOX)
    a.update(kw)
    with pytest.raises(error, match=match):
        rk.rope_write_kv_slot_mapping_quant(a["cs"], a["pos"], a["q"], a["k"], a["v"], a["slots"], a["kc"], a["vc"],
                                            a["ks"], a["vs"], a["qo"], style=a["style"])


@pytest.mark.gpu
@pytest.mark.parametrize("kw,error,match", [
    (dict(lens="cpu"), ValueError, "kv_lens is on cpu"),
    (dict(lens=torch.int64), TypeError, "kv_lens: dtype Long"),
    (dict(q=torch.bfloat16), TypeError, "q: dtype BFloat16"),
    (dict(lse=torch.float16), TypeError, "lse: dtype Half"),
    (dict(table="strided"), ValueError, "page_table must be contiguous"),
    (dict(pool="strided"), ValueError, "kv_cache must be contiguous"),
    (dict(out="strided"), ValueError, "out must be contiguous"),
    (dict(workspace=torch.float32), TypeError, "workspace: dtype Float"),
])
def test_attention_on_the_device(kw, error, match):
    """One argument of another device, type or layout; nothing is launched."""
    a = dict(q=h(3, 1, 4, 64), pool=h(2, 4, 16, 2, 64), prefix=i32(2, 1), table=i32(3, 2, 2), lens=i32(3),
             out=h(3, 1, 4, 64), lse=torch.zeros(3, 1, 4), workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    a = {n: t.to("cuda:0") for n, t in a.items()}
    attention(**a)
    for n, how in kw.items():
        if how == "cpu":
            a[n] = a[n].cpu()
        elif how == "strided":
            a[n] = torch.stack([a[n], a[n]], -1)[..., 0]
        else:
            a[n] = a[n].to(how)
    with pytest.raises(error, match=match):
        attention(**a)
    torch.cuda.synchronize()
